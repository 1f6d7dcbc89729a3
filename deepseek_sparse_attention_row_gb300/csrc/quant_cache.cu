// quant_cache.cu -- writing keys and values into pages of e4m3 codes and
// reading them back: dsa_quant_cache_write and dsa_quant_cache_read of
// include/dsa_quant.h.
#include <cuda_runtime.h>

#include <cmath>

#include "quant.cuh"

namespace dsa {
namespace {

struct WriteArgs {
  QuantPool pool;
  const void* x[2];
  int64_t xt[2], xh[2];  // elements
  int64_t total;
  const int32_t* cu;
  int32_t seqs;
  const int32_t* lens;
};

__device__ __forceinline__ int64_t clamped(int32_t x, int64_t most) {
  return x < 0 ? 0 : (x < most ? x : most);
}

// The last of n + 1 nondecreasing marks that is not above `x`, if mark 0 is not.
template <typename F>
__device__ __forceinline__ int32_t last_upto(int32_t n, int64_t x, F mark) {
  int32_t lo = 0, hi = n;  // mark(lo) <= x, hi: beyond
  while (hi - lo > 1) {
    const int32_t mid = lo + (hi - lo) / 2;
    if (mark(mid) <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

template <typename T>
__device__ __forceinline__ float2 pair(uint32_t two);
template <>
__device__ __forceinline__ float2 pair<__nv_bfloat16>(uint32_t two) {
  return make_float2(__uint_as_float(two << 16), __uint_as_float(two & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 pair<__half>(uint32_t two) {
  return __half22float2(*reinterpret_cast<const __half2*>(&two));
}

__device__ __forceinline__ float finite_size(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.f;
}
__device__ __forceinline__ float nan_for_infinite(float x) {
  return fabsf(x) < INFINITY ? x : NAN;
}

// A block of a sequence that gets new tokens. Sequence s of n tokens touches at
// most n / block + 2 blocks, and floor(cu[s] / block) + 2 s counts that many
// between one sequence and the next: item numbers are found from cu alone.
struct Block {
  int32_t seq, page;  // page -1: nothing to do
  int32_t start;      // its first token
  int32_t from, to;   // the new ones
  int64_t row;        // of the token `from`
};

__device__ __forceinline__ Block find_block(const WriteArgs& a, int64_t item) {
  const int lg = a.pool.block_log2;
  Block b{};
  b.page = -1;
  const int32_t s = last_upto(a.seqs, item, [&](int32_t i) {
    return (clamped(a.cu[i], a.total) >> lg) + 2ll * i;
  });
  const int64_t r0 = clamped(a.cu[s], a.total), r1 = clamped(a.cu[s + 1], a.total);
  const int64_t held = a.lens[s] > 0 ? a.lens[s] : 0, end = held + (r1 - r0);
  const int64_t most = a.pool.max_pages << a.pool.page_log2;
  const int64_t at = item - (r0 >> lg) - 2ll * s;  // below 0: rows in front of the first sequence
  const int64_t start = ((held >> lg) + at) << lg;
  if (at < 0 || r1 <= r0 || start >= end || start >= most) return b;
  b.seq = s;
  b.start = static_cast<int32_t>(start);
  b.from = static_cast<int32_t>(held > start ? held : start);
  b.to = static_cast<int32_t>(end < start + (1ll << lg) ? end : start + (1ll << lg));
  b.row = r0 + b.from - held;
  b.page = quant_page(a.pool, s, b.start);
  return b;
}

constexpr int kWriteWarps = 4;

// A warp for each block, head and one of keys and values.
template <typename T>
__global__ void __launch_bounds__(kWriteWarps * 32) write_kernel(const WriteArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Block b = find_block(a, blockIdx.x);
  if (b.page < 0) return;
  const int parts = a.pool.dim / 8, rows = 32 / parts;  // 8 elements of a lane
  const int row = lane / parts, part = lane % parts;
  for (int w = warp + kWriteWarps * blockIdx.y; w < 2 * a.pool.kv_heads;
       w += kWriteWarps * gridDim.y) {
    const int kv = w & 1, head = w >> 1;
    const char* x = static_cast<const char*>(a.x[kv]) + head * a.xh[kv] * sizeof(T) + part * 16;
    const auto load = [&](int32_t t) {
      return *reinterpret_cast<const uint4*>(
          x + (b.row + t - b.from) * a.xt[kv] * static_cast<int64_t>(sizeof(T)));
    };
    float top = 0.f;
    for (int32_t t = b.from + row; t < b.to && row < rows; t += rows) {
      const uint4 u = load(t);
      for (uint32_t two : {u.x, u.y, u.z, u.w}) {
        const float2 f = pair<T>(two);
        top = fmaxf(top, fmaxf(finite_size(f.x), finite_size(f.y)));
      }
    }
    top = __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(top)));
    uint32_t e = need_exponent(top);
    float* scale = quant_scale(a.pool, kv, b.page, b.start, head);
    if (b.from > b.start) {
      const float was = *scale;
      e = max(e, held_exponent(was));
      __syncwarp();
      if (power(e) != was) {
        for (int32_t t = b.start + row; t < b.from && row < rows; t += rows) {
          uint2* at = reinterpret_cast<uint2*>(quant_code(a.pool, kv, b.page, t, head) + part * 8);
          const uint2 u = *at;
          const auto again = [&](uint32_t four) {
            const float i = inverse_power(e);
            const float2 lo = decode2f(four & 0xffffu), hi = decode2f(four >> 16);
            return encode2(lo.x * was * i, lo.y * was * i) |
                   (encode2(hi.x * was * i, hi.y * was * i) << 16);
          };
          *at = make_uint2(again(u.x), again(u.y));
        }
      }
    }
    if (lane == 0) *scale = power(e);
    const float i = inverse_power(e);
    for (int32_t t = b.from + row; t < b.to && row < rows; t += rows) {
      const uint4 u = load(t);
      const auto code = [&](uint32_t two) {
        const float2 f = pair<T>(two);
        return encode2(nan_for_infinite(f.x) * i, nan_for_infinite(f.y) * i);
      };
      *reinterpret_cast<uint2*>(quant_code(a.pool, kv, b.page, t, head) + part * 8) =
          make_uint2(code(u.x) | (code(u.y) << 16), code(u.z) | (code(u.w) << 16));
    }
  }
}

struct ReadArgs {
  QuantPool pool;
  void* x[2];
  int64_t xt[2], xh[2];
  int64_t total;
  const int32_t* cu;
  int32_t seqs;
};

template <typename T>
__device__ __forceinline__ uint32_t pack(float2 f);
template <>
__device__ __forceinline__ uint32_t pack<__nv_bfloat16>(float2 f) {
  const __nv_bfloat162 h = __float22bfloat162_rn(f);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack<__half>(float2 f) {
  const __half2 h = __float22half2_rn(f);
  return *reinterpret_cast<const uint32_t*>(&h);
}

constexpr int kReadThreads = 256;

// A CTA for each row; a thread for 16 codes.
template <typename T>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const ReadArgs a) {
  const int64_t r = blockIdx.x;
  const int32_t s = last_upto(a.seqs, r, [&](int32_t i) { return clamped(a.cu[i], a.total); });
  const int64_t r0 = clamped(a.cu[s], a.total), r1 = clamped(a.cu[s + 1], a.total);
  if (r < r0 || r >= r1) return;
  const int64_t t = r - r0;
  const int32_t page = t < (a.pool.max_pages << a.pool.page_log2)
                           ? quant_page(a.pool, s, static_cast<int32_t>(t))
                           : -1;
  const int parts = a.pool.dim / 16;
  for (int u = threadIdx.x; u < 2 * a.pool.kv_heads * parts; u += kReadThreads) {
    const int part = u % parts, kv = u / parts & 1, head = u / parts >> 1;
    uint4 c = make_uint4(0, 0, 0, 0);
    float scale = 0.f;
    if (page >= 0) {
      c = *reinterpret_cast<const uint4*>(
          quant_code(a.pool, kv, page, static_cast<int32_t>(t), head) + part * 16);
      scale = *quant_scale(a.pool, kv, page, static_cast<int32_t>(t), head);
    }
    uint4* to = reinterpret_cast<uint4*>(static_cast<T*>(a.x[kv]) + r * a.xt[kv] +
                                         head * a.xh[kv] + part * 16);
    const auto two = [&](uint32_t codes) {
      const float2 f = decode2f(codes);
      return pack<T>(make_float2(f.x * scale, f.y * scale));
    };
    to[0] = make_uint4(two(c.x & 0xffff), two(c.x >> 16), two(c.y & 0xffff), two(c.y >> 16));
    to[1] = make_uint4(two(c.z & 0xffff), two(c.z >> 16), two(c.w & 0xffff), two(c.w >> 16));
  }
}

// What writing and reading check alike: rows of 16-bit elements.
dsa_status check_rows(const void* k, const void* v, int32_t dtype, int64_t total, int64_t k_st,
                      int64_t k_sh, int64_t v_st, int64_t v_sh, const int32_t* cu, int32_t seqs,
                      int32_t kv_heads) {
  if (dtype != DSA_DTYPE_F32 && dtype != DSA_DTYPE_BF16 && dtype != DSA_DTYPE_F16)
    return DSA_EINVAL;
  if (total < 0 || seqs < 0) return DSA_EINVAL;
  if (dtype == DSA_DTYPE_F32 || total > INT32_MAX || seqs >= (1 << 28)) return DSA_EUNSUPPORTED;
  if (total == 0 || seqs == 0 || kv_heads == 0) return DSA_OK;
  if (!k || !v || !cu) return DSA_EINVAL;
  if (!quant_aligned16(k) || !quant_aligned16(v)) return DSA_EUNSUPPORTED;
  for (int64_t s : {k_st, k_sh, v_st, v_sh})
    if (s < 0 || s % 8 != 0) return DSA_EUNSUPPORTED;
  return DSA_OK;
}

}  // namespace
}  // namespace dsa

extern "C" dsa_status dsa_quant_cache_write(
    const void* k, const void* v, int32_t dtype, int64_t total, int32_t kv_heads, int32_t head_dim,
    int64_t k_st, int64_t k_sh, int64_t v_st, int64_t v_sh, const int32_t* cu, int32_t seqs,
    void* k_codes, void* v_codes, int64_t num_pages, int32_t page_size, int32_t block,
    int64_t kc_sn, int64_t kc_st, int64_t kc_sh, int64_t vc_sn, int64_t vc_st, int64_t vc_sh,
    float* k_scales, float* v_scales, int64_t ks_sn, int64_t vs_sn, const int32_t* tables,
    int64_t max_pages, int64_t ld_tables, const int32_t* lens, void* stream) {
  dsa::WriteArgs a{};
  dsa_status st = dsa::quant_pool(a.pool, k_codes, v_codes, k_scales, v_scales, num_pages,
                                  page_size, block, kv_heads, head_dim,
                                  {kc_sn, kc_st, kc_sh, vc_sn, vc_st, vc_sh}, ks_sn, vs_sn, tables,
                                  max_pages, ld_tables, seqs);
  if (st != DSA_OK) return st;
  st = dsa::check_rows(k, v, dtype, total, k_st, k_sh, v_st, v_sh, cu, seqs, kv_heads);
  if (st != DSA_OK) return st;
  if (block > 256) return DSA_EUNSUPPORTED;
  if (total == 0 || seqs == 0 || kv_heads == 0) return DSA_OK;
  if (!lens) return DSA_EINVAL;
  if (max_pages == 0 || num_pages == 0) return DSA_OK;
  a.x[0] = k;
  a.x[1] = v;
  a.xt[0] = k_st;
  a.xt[1] = v_st;
  a.xh[0] = k_sh;
  a.xh[1] = v_sh;
  a.total = total;
  a.cu = cu;
  a.seqs = seqs;
  a.lens = lens;
  const int64_t items = total / block + 2ll * seqs;
  if (items > INT32_MAX) return DSA_EUNSUPPORTED;
  const unsigned ys = static_cast<unsigned>((2ll * kv_heads + dsa::kWriteWarps - 1) /
                                            dsa::kWriteWarps);
  const dim3 grid(static_cast<unsigned>(items), ys < 65535 ? ys : 65535);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == DSA_DTYPE_BF16)
    dsa::write_kernel<__nv_bfloat16><<<grid, dsa::kWriteWarps * 32, 0, s>>>(a);
  else
    dsa::write_kernel<__half><<<grid, dsa::kWriteWarps * 32, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ECUDA;
}

extern "C" dsa_status dsa_quant_cache_read(
    const void* k_codes, const void* v_codes, const float* k_scales, const float* v_scales,
    int64_t num_pages, int32_t page_size, int32_t block, int32_t kv_heads, int32_t head_dim,
    int64_t kc_sn, int64_t kc_st, int64_t kc_sh, int64_t vc_sn, int64_t vc_st, int64_t vc_sh,
    int64_t ks_sn, int64_t vs_sn, const int32_t* tables, int64_t max_pages, int64_t ld_tables,
    const int32_t* cu, int32_t seqs, int64_t total, int32_t dtype, void* k, int64_t k_st,
    int64_t k_sh, void* v, int64_t v_st, int64_t v_sh, void* stream) {
  dsa::ReadArgs a{};
  dsa_status st = dsa::quant_pool(a.pool, k_codes, v_codes, k_scales, v_scales, num_pages,
                                  page_size, block, kv_heads, head_dim,
                                  {kc_sn, kc_st, kc_sh, vc_sn, vc_st, vc_sh}, ks_sn, vs_sn, tables,
                                  max_pages, ld_tables, seqs);
  if (st != DSA_OK) return st;
  st = dsa::check_rows(k, v, dtype, total, k_st, k_sh, v_st, v_sh, cu, seqs, kv_heads);
  if (st != DSA_OK) return st;
  if (total == 0 || seqs == 0 || kv_heads == 0) return DSA_OK;
  a.x[0] = k;
  a.x[1] = v;
  a.xt[0] = k_st;
  a.xt[1] = v_st;
  a.xh[0] = k_sh;
  a.xh[1] = v_sh;
  a.total = total;
  a.cu = cu;
  a.seqs = seqs;
  const unsigned grid = static_cast<unsigned>(total);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == DSA_DTYPE_BF16)
    dsa::read_kernel<__nv_bfloat16><<<grid, dsa::kReadThreads, 0, s>>>(a);
  else
    dsa::read_kernel<__half><<<grid, dsa::kReadThreads, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ECUDA;
}
