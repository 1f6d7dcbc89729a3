// rotary.cu -- rotary positions of queries and keys: the C ABI of
// include/dsa_rotary.h.
//
// A CTA takes a few tokens: it computes the cosines and sines of their positions
// once, into shared memory, and then goes through the heads, a chunk of pairs to
// a thread. Chunks are as wide as alignment lets them be, up to 16 bytes;
// neighbouring threads take neighbouring chunks. The first loads are on their way
// while the angles are computed. (With the angles in registers, computed again
// by every thread, 8192 tokens of 40 heads of 128 took 48 us.)
#include "../../include/dsa_rotary.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

namespace dsa {
namespace {

constexpr int kThreads = 256;

struct RotaryArgs {
  const void *q, *k;
  void *q_out, *k_out;
  int64_t q_st, q_sh, qo_st, qo_sh, k_st, k_sh, ko_st, ko_sh;
  int32_t heads, all_heads;  // all_heads counts those of k too
  int64_t tokens;
  const int32_t* positions;
  const int64_t* turns;
  int32_t pairs;
  int32_t turned, chunks;      // chunks of a head: those of the pairs, and all
  int32_t step, other;         // from chunk to chunk, and to its second half (SPLIT)
  int32_t each, part;          // tokens of a CTA, and heads
  uint32_t by_chunks, by_part;  // ceil(2^32 / chunks) and / part, 0 for 1
  float factor;
  int32_t transpose;
};

// n / d for by = ceil(2^32 / d): exact while n * d is below 2^32.
__device__ __forceinline__ uint32_t quotient(uint32_t n, uint32_t by) {
  return by ? __umulhi(n, by) : n;
}
uint32_t reciprocal(uint32_t d) {
  return d == 1 ? 0 : static_cast<uint32_t>(((1ull << 32) + d - 1) / d);
}

// cos and sin of the angle of position p. The fraction of a turn is exact;
// what is left after the nearest quarter turn, at most an eighth, is rounded
// to fp32 relative to itself, so that both are good to an ulp at any p.
__device__ __forceinline__ float2 cos_sin(int32_t p, int64_t turn, bool transpose) {
  const uint64_t t = static_cast<uint64_t>(static_cast<int64_t>(p)) * static_cast<uint64_t>(turn);
  const uint64_t v = t + (1ull << 61);
  const uint32_t quarter = static_cast<uint32_t>(v >> 62);
  const int32_t rest = static_cast<int32_t>(static_cast<uint32_t>(v >> 30) ^ 0x80000000u);
  float s, c;
  sincospif(static_cast<float>(rest) * 0x1p-33f, &s, &c);  // half turns
  float2 r = quarter & 1 ? make_float2(-s, c) : make_float2(c, s);
  if (quarter & 2) r = make_float2(-r.x, -r.y);
  if (transpose) r.y = -r.y;
  return r;
}

template <typename T>
__device__ __forceinline__ float widen(T x) {
  return static_cast<float>(x);
}
template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half narrow<__half>(float x) {
  return __float2half_rn(x);
}

template <typename T, int V>
struct alignas(V * sizeof(T)) Vec {
  T x[V];
};

// V elements of T at a time. SPLIT: a chunk is V pairs, whose first and second
// elements lie apart; otherwise it is V / 2 pairs of neighbours.
template <typename T, int V, bool SPLIT>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a) {
  constexpr int P = SPLIT ? V : V / 2;  // pairs of a chunk
  constexpr int kAtOnce = SPLIT ? 2 : 4;
  using Chunk = Vec<T, V>;
  // [token][two pairs of a chunk][chunk]: neighbouring threads read neighbours
  extern __shared__ __align__(16) float2 angles[];
  const auto slot = [&](int token, int c, int n) {
    return token * a.pairs + (P > 1 ? ((n >> 1) * a.turned + c) * 2 + (n & 1) : c);
  };
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.each;
  const int tokens = static_cast<int>(min(static_cast<int64_t>(a.each), a.tokens - t0));
  const int first = blockIdx.y * a.part, part = min(a.part, a.all_heads - first);
  const uint32_t units = tokens * a.part * a.chunks;

  Chunk u[kAtOnce], w[SPLIT ? kAtOnce : 1];
  // A unit's token, head and chunk; -1 for none.
  struct Unit {
    int token, head, c;
  };
  const auto unit = [&](uint32_t e) {
    const uint32_t r = quotient(e, a.by_chunks);
    Unit x;
    x.c = static_cast<int>(e - r * a.chunks);
    x.token = static_cast<int>(quotient(r, a.by_part));
    x.head = static_cast<int>(r) - x.token * a.part;
    if (e >= units || x.head >= part) x.token = -1;
    x.head += first;
    return x;
  };
  const auto offset = [&](const Unit& x) {
    return x.c < a.turned ? x.c * a.step : 2 * a.pairs + (x.c - a.turned) * V;
  };
  const auto load = [&](uint32_t e0) {
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const Unit x = unit(e0 + i * kThreads);
      if (x.token < 0) continue;
      const T* from = (x.head < a.heads
                           ? static_cast<const T*>(a.q) + x.head * a.q_sh + (t0 + x.token) * a.q_st
                           : static_cast<const T*>(a.k) + (x.head - a.heads) * a.k_sh +
                                 (t0 + x.token) * a.k_st) +
                      offset(x);
      u[i] = *reinterpret_cast<const Chunk*>(from);
      if constexpr (SPLIT)
        if (x.c < a.turned) w[i] = *reinterpret_cast<const Chunk*>(from + a.other);
    }
  };
  load(threadIdx.x);
  for (int i = threadIdx.x; i < tokens * a.pairs; i += kThreads) {
    const int token = i / a.pairs, pair = i - token * a.pairs, c = pair / P;
    float2 cs = cos_sin(a.positions[t0 + token], a.turns[pair], a.transpose);
    cs.x *= a.factor;
    cs.y *= a.factor;
    angles[slot(token, c, pair - c * P)] = cs;
  }
  __syncthreads();
  for (uint32_t e0 = threadIdx.x;;) {
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const Unit x = unit(e0 + i * kThreads);
      if (x.token < 0) continue;
      T* to = (x.head < a.heads
                   ? static_cast<T*>(a.q_out) + x.head * a.qo_sh + (t0 + x.token) * a.qo_st
                   : static_cast<T*>(a.k_out) + (x.head - a.heads) * a.ko_sh +
                         (t0 + x.token) * a.ko_st) +
              offset(x);
      if (x.c < a.turned) {
#pragma unroll
        for (int n = 0; n < P; ++n) {
          const float2 cs = angles[slot(x.token, x.c, n)];
          T& p = SPLIT ? u[i].x[n] : u[i].x[2 * n];
          T& r = SPLIT ? w[i].x[n] : u[i].x[2 * n + 1];
          const float xa = widen(p), xb = widen(r);
          p = narrow<T>(fmaf(xa, cs.x, -(xb * cs.y)));
          r = narrow<T>(fmaf(xb, cs.x, xa * cs.y));
        }
        if constexpr (SPLIT) *reinterpret_cast<Chunk*>(to + a.other) = w[i];
      }
      *reinterpret_cast<Chunk*>(to) = u[i];
    }
    e0 += kAtOnce * kThreads;
    if (e0 - threadIdx.x >= units) return;
    load(e0);
  }
}

// Units of a CTA (a unit: a chunk of a head), and angles.
constexpr int64_t kUnits = 1024, kAngles = 2048;
constexpr int64_t kCtas = 152 * 4;

template <typename T, int V>
dsa_status launch(RotaryArgs a, int32_t head_dim, bool halves, cudaStream_t stream) {
  // neighbours at addresses that hold no pair whole are taken one by one
  const bool split = halves || V == 1;
  a.turned = split ? a.pairs / V : 2 * a.pairs / V;
  a.chunks = a.turned + (head_dim - 2 * a.pairs) / V;
  a.step = halves ? V : V == 1 ? 2 : V;
  a.other = halves ? a.pairs : 1;
  // As many tokens to a CTA as fill it, while there are CTAs for all SMs; heads
  // are divided where a few tokens have many.
  const int64_t token = static_cast<int64_t>(a.all_heads) * a.chunks;
  int64_t each = kUnits / token, parts = 1;
  if (each > a.tokens / kCtas) each = a.tokens / kCtas;
  if (a.pairs > 0 && each > kAngles / a.pairs) each = kAngles / a.pairs;
  if (each < 1) {
    each = 1;
    parts = (token + kUnits - 1) / kUnits;
    const int64_t few = (kCtas + a.tokens - 1) / a.tokens;  // CTAs that a token may have
    if (parts < few) parts = few < (token + kThreads - 1) / kThreads
                                 ? few
                                 : (token + kThreads - 1) / kThreads;
    if (parts > a.all_heads) parts = a.all_heads;
  }
  a.each = static_cast<int32_t>(each);
  a.part = static_cast<int32_t>((a.all_heads + parts - 1) / parts);
  a.by_chunks = reciprocal(a.chunks);
  a.by_part = reciprocal(a.part);
  const dim3 grid(static_cast<unsigned>((a.tokens + each - 1) / each),
                  static_cast<unsigned>((a.all_heads + a.part - 1) / a.part));
  const size_t smem = static_cast<size_t>(each) * a.pairs * sizeof(float2);
  if (split)
    rotary_kernel<T, V, true><<<grid, kThreads, smem, stream>>>(a);
  else if constexpr (V > 1)
    rotary_kernel<T, V, false><<<grid, kThreads, smem, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ECUDA;
}

// The widest chunk of which `bits` (addresses and steps in bytes, or'ed) and
// the pairs and what is behind them are whole numbers.
template <typename T>
dsa_status launch(const RotaryArgs& a, int32_t head_dim, bool halves, uint64_t bits,
                  cudaStream_t stream) {
  constexpr int e = sizeof(T);
  bits |= static_cast<uint64_t>(halves ? a.pairs : 2 * a.pairs) * e;
  bits |= static_cast<uint64_t>(head_dim - 2 * a.pairs) * e;
  if (bits % 16 == 0) return launch<T, 16 / e>(a, head_dim, halves, stream);
  if (bits % 8 == 0) return launch<T, 8 / e>(a, head_dim, halves, stream);
  if constexpr (e == 2)
    if (bits % 4 == 0) return launch<T, 2>(a, head_dim, halves, stream);
  return launch<T, 1>(a, head_dim, halves, stream);
}

}  // namespace
}  // namespace dsa

extern "C" dsa_status dsa_rotary(const void* q, void* q_out, int32_t heads, int64_t q_st,
                                 int64_t q_sh, int64_t qo_st, int64_t qo_sh, const void* k,
                                 void* k_out, int32_t kv_heads, int64_t k_st, int64_t k_sh,
                                 int64_t ko_st, int64_t ko_sh, int32_t dtype, int64_t tokens,
                                 int32_t head_dim, const int32_t* positions, const int64_t* turns,
                                 int32_t pairs, int32_t interleaved, float factor,
                                 int32_t transpose, void* stream) {
  if (dtype != DSA_DTYPE_F32 && dtype != DSA_DTYPE_BF16 && dtype != DSA_DTYPE_F16)
    return DSA_EINVAL;
  if (heads < 0 || kv_heads < 0 || tokens < 0 || head_dim < 0 || pairs < 0 ||
      pairs > head_dim / 2 || !std::isfinite(factor))
    return DSA_EINVAL;
  const int64_t all = static_cast<int64_t>(heads) + kv_heads;
  const int64_t strides[] = {q_st, q_sh, qo_st, qo_sh, k_st, k_sh, ko_st, ko_sh};
  for (int i = heads > 0 ? 0 : 4; i < (kv_heads > 0 ? 8 : 4); ++i)
    if (strides[i] < 0) return DSA_EINVAL;
  if (tokens > INT32_MAX || head_dim > 4096 || all > 65535)
    return DSA_EUNSUPPORTED;
  if (tokens == 0 || head_dim == 0 || all == 0) return DSA_OK;
  if ((heads > 0 && (!q || !q_out)) || (kv_heads > 0 && (!k || !k_out)) ||
      (pairs > 0 && (!positions || !turns)))
    return DSA_EINVAL;
  const uint64_t e = dtype == DSA_DTYPE_F32 ? 4 : 2;
  uint64_t bits = 0;
  if (heads > 0)
    bits |= reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(q_out) |
            static_cast<uint64_t>(q_st | q_sh | qo_st | qo_sh) * e;
  if (kv_heads > 0)
    bits |= reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(k_out) |
            static_cast<uint64_t>(k_st | k_sh | ko_st | ko_sh) * e;
  if (bits % e != 0) return DSA_EINVAL;
  dsa::RotaryArgs a{};
  a.q = q;
  a.k = k;
  a.q_out = q_out;
  a.k_out = k_out;
  a.q_st = q_st;
  a.q_sh = q_sh;
  a.qo_st = qo_st;
  a.qo_sh = qo_sh;
  a.k_st = k_st;
  a.k_sh = k_sh;
  a.ko_st = ko_st;
  a.ko_sh = ko_sh;
  a.heads = heads;
  a.all_heads = static_cast<int32_t>(all);
  a.tokens = tokens;
  a.positions = positions;
  a.turns = turns;
  a.pairs = pairs;
  a.factor = factor;
  a.transpose = transpose != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool halves = interleaved == 0;
  if (dtype == DSA_DTYPE_F32) return dsa::launch<float>(a, head_dim, halves, bits, s);
  if (dtype == DSA_DTYPE_BF16) return dsa::launch<__nv_bfloat16>(a, head_dim, halves, bits, s);
  return dsa::launch<__half>(a, head_dim, halves, bits, s);
}
