// quant.cuh -- what the operators on the 8-bit cache share: the pool of pages
// as the kernels see it, and the e4m3 codes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "../../include/dsa_quant.h"

namespace dsa {

// Pages of codes and scales (include/dsa_quant.h), keys first.
struct QuantPool {
  uint8_t* codes[2];
  float* scales[2];
  int64_t sn[2], st[2], sh[2];  // bytes
  int64_t ssn[2];               // floats
  int64_t num_pages;
  int32_t page_log2, block_log2;
  int32_t kv_heads, dim;
  const int32_t* tables;
  int64_t max_pages, ld_tables;
};

constexpr int32_t kMaxKvHeads = 1 << 20;

inline bool quant_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int32_t floor_log2(int64_t n) {
  int32_t l = 0;
  while ((n >> (l + 1)) > 0) ++l;
  return l;
}

// Fills `p` from a call's arguments; the status of what is wrong with them.
inline dsa_status quant_pool(QuantPool& p, const dsa_quant_pages* pages, int64_t seqs) {
  if (!pages) return DSA_EINVAL;
  const dsa_quant_pages& x = *pages;
  if (x.num_pages < 0 || x.page_size < 1 || x.block < 1 || x.kv_heads < 0 || x.head_dim < 1 ||
      x.max_pages < 0 || x.ld_tables < x.max_pages || x.ks_sn < 0 || x.vs_sn < 0)
    return DSA_EINVAL;
  if (x.page_size % x.block != 0) return DSA_EINVAL;
  if (x.num_pages > INT32_MAX || x.max_pages > INT32_MAX || x.page_size < 16 ||
      (x.page_size & (x.page_size - 1)) != 0 || (x.block & (x.block - 1)) != 0 ||
      x.max_pages * x.page_size > INT32_MAX || x.head_dim > 128 || x.head_dim % 16 != 0 ||
      x.kv_heads > kMaxKvHeads)
    return DSA_EUNSUPPORTED;
  if (x.num_pages > 0 && (!x.k_codes || !x.v_codes || !x.k_scales || !x.v_scales))
    return DSA_EINVAL;
  if (x.max_pages > 0 && seqs > 0 && !x.tables) return DSA_EINVAL;
  if (!quant_aligned16(x.k_codes) || !quant_aligned16(x.v_codes)) return DSA_EUNSUPPORTED;
  if (((reinterpret_cast<uintptr_t>(x.k_scales) | reinterpret_cast<uintptr_t>(x.v_scales)) & 3u) !=
      0)
    return DSA_EUNSUPPORTED;
  for (int64_t s : {x.kc_sn, x.kc_st, x.kc_sh, x.vc_sn, x.vc_st, x.vc_sh})
    if (s < 0 || s % 16 != 0) return DSA_EUNSUPPORTED;
  p.codes[0] = static_cast<uint8_t*>(x.k_codes);
  p.codes[1] = static_cast<uint8_t*>(x.v_codes);
  p.scales[0] = x.k_scales;
  p.scales[1] = x.v_scales;
  p.sn[0] = x.kc_sn;
  p.st[0] = x.kc_st;
  p.sh[0] = x.kc_sh;
  p.sn[1] = x.vc_sn;
  p.st[1] = x.vc_st;
  p.sh[1] = x.vc_sh;
  p.ssn[0] = x.ks_sn;
  p.ssn[1] = x.vs_sn;
  p.num_pages = x.num_pages;
  p.page_log2 = floor_log2(x.page_size);
  p.block_log2 = floor_log2(x.block);
  p.kv_heads = x.kv_heads;
  p.dim = x.head_dim;
  p.tables = x.tables;
  p.max_pages = x.max_pages;
  p.ld_tables = x.ld_tables;
  return DSA_OK;
}

// The page of token `t` of sequence `s` (t within the table); -1 for none.
__device__ __forceinline__ int32_t quant_page(const QuantPool& p, int64_t s, int32_t t) {
  const int32_t id = p.tables[s * p.ld_tables + (t >> p.page_log2)];
  return id >= 0 && id < p.num_pages ? id : -1;
}

__device__ __forceinline__ uint8_t* quant_code(const QuantPool& p, int kv, int32_t page, int32_t t,
                                               int32_t head) {
  const int32_t in = t & ((1 << p.page_log2) - 1);
  return p.codes[kv] + page * p.sn[kv] + in * p.st[kv] + head * p.sh[kv];
}

__device__ __forceinline__ float* quant_scale(const QuantPool& p, int kv, int32_t page, int32_t t,
                                              int32_t head) {
  const int32_t in = (t & ((1 << p.page_log2) - 1)) >> p.block_log2;
  return p.scales[kv] + page * p.ssn[kv] + static_cast<int64_t>(in) * p.kv_heads + head;
}

// ---- codes -----------------------------------------------------------------

// Two codes from two floats (the first one in the low byte), to nearest even,
// what passes 448 becomes 448; NaN for NaN.
__device__ __forceinline__ uint32_t encode2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two codes (of the low 16 bits) as fp16: exact.
__device__ __forceinline__ uint32_t decode2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 x;\n\tcvt.u16.u32 x, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\t}"
      : "=r"(r)
      : "r"(two));
  return r;
}
__device__ __forceinline__ float2 decode2f(uint32_t two) {
  const uint32_t h = decode2(two);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The least power of two, from 2^-126 to 2^126, whose product with 1.mantissa *
// 2^down is not below x (x >= 0 and finite), as biased exponent bits.
__device__ __forceinline__ uint32_t power_exponent(float x, uint32_t mantissa, int down) {
  const int e = static_cast<int>((__float_as_uint(x) + (0x7fffffu - mantissa)) >> 23) - down;
  return static_cast<uint32_t>(e < 1 ? 1 : (e > 253 ? 253 : e));
}
// That of a block whose largest finite value is `top`: 448 = 1.75 * 2^8.
__device__ __forceinline__ uint32_t need_exponent(float top) {
  return power_exponent(top, 0x600000u, 8);
}
// The same for an old scale.
__device__ __forceinline__ uint32_t held_exponent(float scale) {
  return scale > 0.f ? power_exponent(fminf(scale, 0x1p126f), 0u, 0) : 1u;
}
__device__ __forceinline__ float power(uint32_t exponent) {
  return __uint_as_float(exponent << 23);
}
// 1 / power(exponent); exponents of 1 to 253.
__device__ __forceinline__ float inverse_power(uint32_t exponent) {
  return __uint_as_float((254u - exponent) << 23);
}

}  // namespace dsa
