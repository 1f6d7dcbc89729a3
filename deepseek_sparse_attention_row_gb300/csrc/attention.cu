// attention.cu -- prompt attention and shared-prefix decode attention: the C
// ABI of include/dsa_attention.h.
//
// Per query row, over the keys that it sees (c = scale * log2 e):
//   x_j = c <q, k_j>,  m = max x_j,  l = sum 2^(x_j - m),
//   out = (sum 2^(x_j - m) v_j) / l,  lse = m + log2 l.
// One warp takes one row and walks its keys 32 at a time with a running
// maximum and sum: a lane forms the product of one key with the row (kept in
// shared memory as fp32), then every lane adds its dimensions of the 32
// values.
#include "../../include/dsa_attention.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

namespace dsa {
namespace {

constexpr int kMaxHeadDim = 128;
constexpr int kMaxGroup = 128;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f(float x) { return __float2half_rn(x); }

// Where key (or value) j of one row's sequence lies: nullptr when no page
// holds it.
template <typename T>
struct Packed {
  const T* base;
  int64_t st;
  __device__ const T* at(int64_t j) const { return base + j * st; }
};
template <typename T>
struct Paged {
  const T* base;  // head's offset included
  int64_t sn, st;
  const int32_t* prefix;
  int64_t prefix_len;
  const int32_t* table;
  int64_t num_pages;
  int32_t page_size;
  __device__ const T* at(int64_t j) const {
    const int64_t p = j / page_size;
    const int32_t id = j < prefix_len ? prefix[p] : table[p];
    if (id < 0 || id >= num_pages) return nullptr;
    return base + id * sn + (j % page_size) * st;
  }
};

// One warp, one row: q in qs (fp32, shared memory), keys [0, n).
template <typename T, typename KAt, typename VAt>
__device__ void attend_row(const float* qs, int dim, const KAt& ks, const VAt& vs, int64_t n,
                           float c, T* out, float* lse) {
  const int lane = threadIdx.x & 31;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};  // dimensions lane + 32 i
  float m = -INFINITY, l = 0.f;
  for (int64_t j0 = 0; j0 < n; j0 += 32) {
    float x = -INFINITY;
    const T* k = j0 + lane < n ? ks.at(j0 + lane) : nullptr;
    if (k) {
      x = 0.f;
      for (int d = 0; d < dim; ++d) x = fmaf(qs[d], to_f(k[d]), x);
      x *= c;
    }
    float mx = x;
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
    const float m_new = fmaxf(m, mx);
    const float base = m_new == -INFINITY ? 0.f : m_new;
    const float keep = exp2f(m - base);
    const float p = exp2f(x - base);  // 0 for keys that are not seen
    float sum = p;
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    l = l * keep + sum;
    m = m_new;
    for (int i = 0; i < 4; ++i) acc[i] *= keep;
    const int32_t cnt = static_cast<int32_t>(n - j0 < 32 ? n - j0 : 32);
    for (int32_t jj = 0; jj < cnt; ++jj) {
      const float pj = __shfl_sync(~0u, p, jj);
      const T* v = vs.at(j0 + jj);
      if (!v) continue;
      for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < dim) acc[i] = fmaf(pj, to_f(v[lane + 32 * i]), acc[i]);
    }
  }
  // l is 0 only where no key was seen (or every weight is 0 by x = -inf)
  const float inv = l == 0.f ? 0.f : 1.f / l;
  for (int i = 0; i < 4; ++i)
    if (lane + 32 * i < dim) out[lane + 32 * i] = from_f<T>(l == 0.f ? 0.f : acc[i] * inv);
  if (lse && lane == 0) *lse = l == 0.f ? -INFINITY : m + log2f(l);
}

struct PromptArgs {
  const void *q, *k, *v;
  int64_t total_q, total_k;
  int32_t heads, kv_heads, dim;
  int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh;
  const int32_t *cu_q, *cu_k;
  int32_t seqs, causal;
  float c;
  void* out;
  int64_t o_st, o_sh;
  float* lse;
  int64_t l_st, l_sh;
};

__device__ __forceinline__ int64_t clamped(int32_t x, int64_t top) {
  return x < 0 ? 0 : (x > top ? top : x);
}

constexpr int kWarps = 8;

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) prompt_kernel(const PromptArgs a) {
  __shared__ float qs[kWarps][kMaxHeadDim];
  float* mine = qs[threadIdx.x >> 5];
  const int lane = threadIdx.x & 31;
  const int64_t rows = a.total_q * a.heads;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); r < rows;
       r += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int64_t t = r / a.heads;
    const int32_t h = static_cast<int32_t>(r % a.heads);
    // the sequence of token t: the last one that starts at or before it
    int32_t lo = 0, hi = a.seqs;  // cu_q[lo] <= t < cu_q[hi]
    if (t < clamped(a.cu_q[0], a.total_q) || t >= clamped(a.cu_q[a.seqs], a.total_q)) continue;
    while (hi - lo > 1) {
      const int32_t mid = (lo + hi) >> 1;
      if (clamped(a.cu_q[mid], a.total_q) <= t) lo = mid; else hi = mid;
    }
    const int64_t q0 = clamped(a.cu_q[lo], a.total_q), q1 = clamped(a.cu_q[lo + 1], a.total_q);
    const int64_t k0 = clamped(a.cu_k[lo], a.total_k);
    int64_t n = clamped(a.cu_k[lo + 1], a.total_k) - k0;
    if (n < 0) n = 0;
    if (a.causal) {
      const int64_t lim = t - q0 + 1 + n - (q1 - q0);
      n = lim < n ? (lim < 0 ? 0 : lim) : n;
    }
    const int64_t kh = h / (a.heads / a.kv_heads);
    const T* q = static_cast<const T*>(a.q) + t * a.q_st + h * a.q_sh;
    __syncwarp();
    for (int d = lane; d < a.dim; d += 32) mine[d] = to_f(q[d]);
    __syncwarp();
    const Packed<T> ks{static_cast<const T*>(a.k) + k0 * a.k_st + kh * a.k_sh, a.k_st};
    const Packed<T> vs{static_cast<const T*>(a.v) + k0 * a.v_st + kh * a.v_sh, a.v_st};
    attend_row<T>(mine, a.dim, ks, vs, n, a.c, static_cast<T*>(a.out) + t * a.o_st + h * a.o_sh,
                  a.lse ? a.lse + t * a.l_st + h * a.l_sh : nullptr);
  }
}

struct SharedArgs {
  const void *q, *k, *v;
  int64_t batch;
  int32_t heads, kv_heads, dim;
  int64_t num_pages;
  int32_t page_size;
  int64_t q_sb, q_sh, k_sn, k_st, k_sh, v_sn, v_st, v_sh;
  const int32_t* prefix_pages;
  int64_t prefix_len;
  const int32_t* tables;
  int64_t max_pages, ld_tables;
  const int32_t* lens;
  float c;
  void* out;
  int64_t o_sb, o_sh;
  float* lse;
  int64_t l_sb, l_sh;
};

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) shared_kernel(const SharedArgs a) {
  __shared__ float qs[kWarps][kMaxHeadDim];
  float* mine = qs[threadIdx.x >> 5];
  const int lane = threadIdx.x & 31;
  const int64_t rows = a.batch * a.heads;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); r < rows;
       r += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int64_t b = r / a.heads, h = r % a.heads;
    const int64_t kh = h / (a.heads / a.kv_heads);
    const int64_t n = clamped(a.lens[b], a.max_pages * a.page_size);
    const T* q = static_cast<const T*>(a.q) + b * a.q_sb + h * a.q_sh;
    __syncwarp();
    for (int d = lane; d < a.dim; d += 32) mine[d] = to_f(q[d]);
    __syncwarp();
    const int32_t* table = a.tables + b * a.ld_tables;
    const Paged<T> ks{static_cast<const T*>(a.k) + kh * a.k_sh, a.k_sn, a.k_st, a.prefix_pages,
                      a.prefix_len, table, a.num_pages, a.page_size};
    const Paged<T> vs{static_cast<const T*>(a.v) + kh * a.v_sh, a.v_sn, a.v_st, a.prefix_pages,
                      a.prefix_len, table, a.num_pages, a.page_size};
    attend_row<T>(mine, a.dim, ks, vs, n, a.c, static_cast<T*>(a.out) + b * a.o_sb + h * a.o_sh,
                  a.lse ? a.lse + b * a.l_sb + h * a.l_sh : nullptr);
  }
}

unsigned grid_for(int64_t rows) {
  const int64_t want = (rows + kWarps - 1) / kWarps;
  return static_cast<unsigned>(want < 4096 ? want : 4096);
}

// Sizes and scale that both operators share.
dsa_status check_common(int32_t dtype, int64_t tokens, int32_t heads, int32_t kv_heads,
                        int32_t head_dim, float scale) {
  if (dtype != DSA_DTYPE_F32 && dtype != DSA_DTYPE_BF16 && dtype != DSA_DTYPE_F16)
    return DSA_EINVAL;
  if (tokens < 0 || heads < 0 || kv_heads < 1 || heads % kv_heads != 0 || head_dim < 1)
    return DSA_EINVAL;
  if (!(scale > 0.f) || !std::isfinite(scale)) return DSA_EINVAL;
  if (dtype == DSA_DTYPE_F32 || head_dim > kMaxHeadDim || head_dim % 8 != 0 ||
      heads / kv_heads > kMaxGroup || tokens > INT32_MAX)
    return DSA_EUNSUPPORTED;
  return DSA_OK;
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
    int64_t l_st, int64_t l_sh, void* stream) {
  if (total_k < 0 || seqs < 0) return DSA_EINVAL;
  const dsa_status st = dsa::check_common(dtype, total_q, heads, kv_heads, head_dim, scale);
  if (st != DSA_OK) return st;
  if (total_k > INT32_MAX) return DSA_EUNSUPPORTED;
  if (total_q == 0 || heads == 0 || seqs == 0) return DSA_OK;
  if (!q || !out || !cu_q || !cu_k || (total_k > 0 && (!k || !v))) return DSA_EINVAL;
  if (!dsa::aligned16(q) || !dsa::aligned16(k) || !dsa::aligned16(v) || !dsa::aligned16(out) ||
      !dsa::by8(q_st, q_sh) || !dsa::by8(k_st, k_sh) || !dsa::by8(v_st, v_sh) ||
      !dsa::by8(o_st, o_sh))
    return DSA_EUNSUPPORTED;
  const dsa::PromptArgs a{q,    k,    v,    total_q, total_k, heads, kv_heads, head_dim,
                          q_st, q_sh, k_st, k_sh,    v_st,    v_sh,  cu_q,     cu_k,
                          seqs, causal, scale * dsa::kLog2e, out, o_st, o_sh, lse, l_st, l_sh};
  const unsigned grid = dsa::grid_for(total_q * heads);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == DSA_DTYPE_BF16)
    dsa::prompt_kernel<__nv_bfloat16><<<grid, dsa::kWarps * 32, 0, s>>>(a);
  else
    dsa::prompt_kernel<__half><<<grid, dsa::kWarps * 32, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ECUDA;
}

extern "C" size_t dsa_shared_prefix_workspace_bytes(int64_t batch, int32_t heads,
                                                    int32_t kv_heads, int32_t head_dim,
                                                    int64_t prefix_len, int64_t max_pages,
                                                    int32_t page_size) {
  (void)batch, (void)heads, (void)kv_heads, (void)head_dim;
  (void)prefix_len, (void)max_pages, (void)page_size;
  return 0;
}

extern "C" dsa_status dsa_shared_prefix_attention(
    const void* q, const void* k_pages, const void* v_pages, int32_t dtype, int64_t batch,
    int32_t heads, int32_t kv_heads, int32_t head_dim, int64_t num_pages, int32_t page_size,
    int64_t q_sb, int64_t q_sh, int64_t k_sn, int64_t k_st, int64_t k_sh, int64_t v_sn,
    int64_t v_st, int64_t v_sh, const int32_t* prefix_pages, int64_t prefix_len,
    const int32_t* tables, int64_t max_pages, int64_t ld_tables, const int32_t* lens, float scale,
    void* out, int64_t o_sb, int64_t o_sh, float* lse, int64_t l_sb, int64_t l_sh,
    void* workspace, size_t workspace_bytes, void* stream) {
  (void)workspace, (void)workspace_bytes;
  if (num_pages < 0 || page_size < 1 || max_pages < 0 || ld_tables < max_pages || prefix_len < 0)
    return DSA_EINVAL;
  const dsa_status st = dsa::check_common(dtype, batch, heads, kv_heads, head_dim, scale);
  if (st != DSA_OK) return st;
  if (num_pages > INT32_MAX || max_pages > INT32_MAX || page_size < 16 ||
      (page_size & (page_size - 1)) != 0 || max_pages * page_size > INT32_MAX)
    return DSA_EUNSUPPORTED;
  if (prefix_len % page_size != 0 || prefix_len > max_pages * page_size) return DSA_EINVAL;
  if (batch == 0 || heads == 0) return DSA_OK;
  if (!q || !out || !lens || (max_pages > 0 && !tables) || (prefix_len > 0 && !prefix_pages) ||
      (num_pages > 0 && (!k_pages || !v_pages)))
    return DSA_EINVAL;
  if (!dsa::aligned16(q) || !dsa::aligned16(k_pages) || !dsa::aligned16(v_pages) ||
      !dsa::aligned16(out) || !dsa::by8(q_sb, q_sh) || !dsa::by8(k_sn, k_st, k_sh) ||
      !dsa::by8(v_sn, v_st, v_sh) || !dsa::by8(o_sb, o_sh))
    return DSA_EUNSUPPORTED;
  const dsa::SharedArgs a{q,         k_pages, v_pages, batch, heads,  kv_heads, head_dim,
                          num_pages, page_size, q_sb,  q_sh,  k_sn,   k_st,     k_sh,
                          v_sn,      v_st,    v_sh,    prefix_pages, prefix_len, tables,
                          max_pages, ld_tables, lens,  scale * dsa::kLog2e, out, o_sb, o_sh,
                          lse,       l_sb,    l_sh};
  const unsigned grid = dsa::grid_for(batch * heads);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == DSA_DTYPE_BF16)
    dsa::shared_kernel<__nv_bfloat16><<<grid, dsa::kWarps * 32, 0, s>>>(a);
  else
    dsa::shared_kernel<__half><<<grid, dsa::kWarps * 32, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ECUDA;
}
