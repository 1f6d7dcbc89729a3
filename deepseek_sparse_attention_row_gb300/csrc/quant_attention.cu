// quant_attention.cu -- attention of single tokens over pages of e4m3 codes:
// dsa_quant_attention of include/dsa_quant.h.
#include <cuda_runtime.h>

#include <cmath>

#include "quant.cuh"

namespace dsa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

struct AttnArgs {
  QuantPool pool;
  const void* q;
  int64_t q_sb, q_sh;
  int32_t heads, group;
  const int32_t* lens;
  float c;  // scale * log2 e
  void* out;
  int64_t o_sb, o_sh;
  float* lse;
  int64_t l_sb, l_sh;
};

constexpr int kWarps = 4;

// A CTA for each sequence and head; its warps take every fourth token.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) attention_kernel(const AttnArgs a) {
  __shared__ float part[kWarps][130];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t b = blockIdx.x / a.heads;
  const int h = blockIdx.x % a.heads, head = h / a.group, d = lane * 4;
  const bool mine = d < a.pool.dim;
  float q[4] = {}, o[4] = {};
  if (mine) {
    const T* row = static_cast<const T*>(a.q) + b * a.q_sb + h * a.q_sh + d;
    for (int i = 0; i < 4; ++i) q[i] = static_cast<float>(row[i]);
  }
  int64_t n = a.lens[b];
  const int64_t most = a.pool.max_pages << a.pool.page_log2;
  n = n < 0 ? 0 : (n < most ? n : most);
  float m = -INFINITY, l = 0.f;
  for (int32_t t = warp; t < n; t += kWarps) {
    const int32_t page = quant_page(a.pool, b, t);
    if (page < 0) continue;
    uint32_t kc = 0, vc = 0;
    if (mine) {
      kc = *reinterpret_cast<const uint32_t*>(quant_code(a.pool, 0, page, t, head) + d);
      vc = *reinterpret_cast<const uint32_t*>(quant_code(a.pool, 1, page, t, head) + d);
    }
    const float2 k0 = decode2f(kc & 0xffff), k1 = decode2f(kc >> 16);
    float x = q[0] * k0.x + q[1] * k0.y + q[2] * k1.x + q[3] * k1.y;
    for (int i = 16; i; i >>= 1) x += __shfl_xor_sync(~0u, x, i);
    x *= a.c * *quant_scale(a.pool, 0, page, t, head);
    const float top = x > m ? x : m, base = top == -INFINITY ? 0.f : top;
    const float keep = exp2f(m - base), p = exp2f(x - base);
    const float pv = p * *quant_scale(a.pool, 1, page, t, head);
    const float2 v0 = decode2f(vc & 0xffff), v1 = decode2f(vc >> 16);
    l = l * keep + p;
    o[0] = o[0] * keep + pv * v0.x;
    o[1] = o[1] * keep + pv * v0.y;
    o[2] = o[2] * keep + pv * v1.x;
    o[3] = o[3] * keep + pv * v1.y;
    m = top;
  }
  for (int i = 0; i < 4; ++i)
    if (mine) part[warp][d + i] = o[i];
  if (lane == 0) {
    part[warp][128] = m;
    part[warp][129] = l;
  }
  __syncthreads();
  float top = -INFINITY;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, part[w][128]);
  const float base = top == -INFINITY ? 0.f : top;
  float sum = 0.f, out = 0.f;
  for (int w = 0; w < kWarps; ++w) {
    const float f = exp2f(part[w][128] - base);
    sum += f * part[w][129];
    if (threadIdx.x < a.pool.dim) out += f * part[w][threadIdx.x];
  }
  if (threadIdx.x < a.pool.dim)
    static_cast<T*>(a.out)[b * a.o_sb + h * a.o_sh + threadIdx.x] =
        static_cast<T>(sum == 0.f ? 0.f : out / sum);
  if (threadIdx.x == 0 && a.lse) a.lse[b * a.l_sb + h * a.l_sh] = base + log2f(sum);
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
  return 0;
}

extern "C" dsa_status dsa_quant_attention(
    const void* q, int32_t dtype, int64_t batch, int32_t heads, int32_t kv_heads, int32_t head_dim,
    int64_t q_sb, int64_t q_sh, const void* k_codes, const void* v_codes, const float* k_scales,
    const float* v_scales, int64_t num_pages, int32_t page_size, int32_t block, int64_t kc_sn,
    int64_t kc_st, int64_t kc_sh, int64_t vc_sn, int64_t vc_st, int64_t vc_sh, int64_t ks_sn,
    int64_t vs_sn, const int32_t* tables, int64_t max_pages, int64_t ld_tables,
    const int32_t* lens, float scale, void* out, int64_t o_sb, int64_t o_sh, float* lse,
    int64_t l_sb, int64_t l_sh, void* workspace, size_t workspace_bytes, void* stream) {
  if (dtype != DSA_DTYPE_F32 && dtype != DSA_DTYPE_BF16 && dtype != DSA_DTYPE_F16)
    return DSA_EINVAL;
  if (!(scale > 0.f) || !std::isfinite(scale * dsa::kLog2e)) return DSA_EINVAL;
  dsa::AttnArgs a{};
  dsa_status st = dsa::quant_pool(a.pool, k_codes, v_codes, k_scales, v_scales, num_pages,
                                  page_size, block, kv_heads, head_dim,
                                  {kc_sn, kc_st, kc_sh, vc_sn, vc_st, vc_sh}, ks_sn, vs_sn, tables,
                                  max_pages, ld_tables, batch);
  if (st != DSA_OK) return st;
  st = dsa::check_sizes(batch, heads, kv_heads);
  if (st != DSA_OK) return st;
  if (dtype == DSA_DTYPE_F32) return DSA_EUNSUPPORTED;
  if (batch == 0 || heads == 0) return DSA_OK;
  if (!q || !out || !lens) return DSA_EINVAL;
  if (!dsa::quant_aligned16(q) || !dsa::quant_aligned16(out)) return DSA_EUNSUPPORTED;
  for (int64_t s : {q_sb, q_sh, o_sb, o_sh})
    if (s < 0 || s % 8 != 0) return DSA_EUNSUPPORTED;
  if (num_pages == 0) a.pool.max_pages = 0;
  a.q = q;
  a.q_sb = q_sb;
  a.q_sh = q_sh;
  a.heads = heads;
  a.group = heads / kv_heads;
  a.lens = lens;
  a.c = scale * dsa::kLog2e;
  a.out = out;
  a.o_sb = o_sb;
  a.o_sh = o_sh;
  a.lse = lse;
  a.l_sb = l_sb;
  a.l_sh = l_sh;
  const unsigned grid = static_cast<unsigned>(batch * heads);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == DSA_DTYPE_BF16)
    dsa::attention_kernel<__nv_bfloat16><<<grid, dsa::kWarps * 32, 0, s>>>(a);
  else
    dsa::attention_kernel<__half><<<grid, dsa::kWarps * 32, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ECUDA;
}
