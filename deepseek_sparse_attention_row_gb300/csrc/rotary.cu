// rotary.cu -- rotary positions of queries and keys: the C ABI of
// include/dsa_rotary.h.
//
// A thread owns one chunk of pairs of one token and goes through heads with
// it: the angle is the same for all heads, so that cosines and sines are
// computed once and stay in registers. Chunks are as wide as alignment lets
// them be, up to 16 bytes; neighbouring threads take neighbouring chunks.
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
  uint32_t tokens;
  const int32_t* positions;
  const int64_t* turns;
  int32_t pairs;
  int32_t turned;          // chunks of a head: those of the pairs,
  uint32_t chunks, lanes;  // all, and threads that share a token's chunk
  float factor;
  int32_t transpose;
};

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

// This thread's token, chunk and first head.
__device__ __forceinline__ bool place(const RotaryArgs& a, uint32_t& t, int& c, int& first) {
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x, j = i / a.chunks;
  t = j / a.lanes;
  c = static_cast<int>(i - j * a.chunks);
  first = static_cast<int>(j - t * a.lanes);
  return t < a.tokens;
}

template <typename T, int V>
struct alignas(V * sizeof(T)) Vec {
  T x[V];
};

// V elements of T at a time. HALVES: a chunk is V pairs (V elements from each
// half); otherwise it is V / 2 neighbouring pairs.
template <typename T, int V, bool HALVES>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a) {
  constexpr int P = HALVES ? V : V / 2;  // pairs of a chunk
  using Chunk = Vec<T, V>;
  uint32_t t;
  int c, first;
  if (!place(a, t, c, first)) return;
  const bool turned = c < a.turned;
  // where the chunk lies, and the other half of its pairs
  const int at = turned ? c * V : 2 * a.pairs + (c - a.turned) * V;
  const int other = HALVES && turned ? a.pairs : 0;
  float2 cs[P];
#pragma unroll
  for (int n = 0; n < P; ++n) cs[n] = make_float2(0.f, 0.f);
  if (turned) {
    const int32_t p = a.positions[t];
#pragma unroll
    for (int n = 0; n < P; ++n) {
      cs[n] = cos_sin(p, a.turns[c * P + n], a.transpose);
      cs[n].x *= a.factor;
      cs[n].y *= a.factor;
    }
  }
  const T* q = static_cast<const T*>(a.q) + t * a.q_st + at;
  const T* k = static_cast<const T*>(a.k) + t * a.k_st + at;
  T* qo = static_cast<T*>(a.q_out) + t * a.qo_st + at;
  T* ko = static_cast<T*>(a.k_out) + t * a.ko_st + at;
  // Outputs may be inputs, so that loads would wait for the stores before them:
  // those of kAtOnce heads come first.
  constexpr int kAtOnce = HALVES ? 4 : 8;
  for (int h0 = first; h0 < a.all_heads; h0 += kAtOnce * a.lanes) {
    Chunk u[kAtOnce], w[HALVES ? kAtOnce : 1];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int h = h0 + i * a.lanes;
      if (h >= a.all_heads) continue;
      const T* x = h < a.heads ? q + h * a.q_sh : k + (h - a.heads) * a.k_sh;
      u[i] = *reinterpret_cast<const Chunk*>(x);
      if constexpr (HALVES) w[i] = *reinterpret_cast<const Chunk*>(x + other);
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int h = h0 + i * a.lanes;
      if (h >= a.all_heads) continue;
      T* y = h < a.heads ? qo + h * a.qo_sh : ko + (h - a.heads) * a.ko_sh;
      if (turned) {
        if constexpr (HALVES) {
#pragma unroll
          for (int n = 0; n < V; ++n) {
            const float xa = widen(u[i].x[n]), xb = widen(w[i].x[n]);
            u[i].x[n] = narrow<T>(fmaf(xa, cs[n].x, -(xb * cs[n].y)));
            w[i].x[n] = narrow<T>(fmaf(xb, cs[n].x, xa * cs[n].y));
          }
          *reinterpret_cast<Chunk*>(y + other) = w[i];
        } else {
#pragma unroll
          for (int n = 0; n < P; ++n) {
            const float xa = widen(u[i].x[2 * n]), xb = widen(u[i].x[2 * n + 1]);
            u[i].x[2 * n] = narrow<T>(fmaf(xa, cs[n].x, -(xb * cs[n].y)));
            u[i].x[2 * n + 1] = narrow<T>(fmaf(xb, cs[n].x, xa * cs[n].y));
          }
        }
      }
      *reinterpret_cast<Chunk*>(y) = u[i];
    }
  }
}

// Neighbouring pairs at addresses that hold no pair whole, element by element.
template <typename T>
__global__ void __launch_bounds__(kThreads) rotary_pairs_kernel(const RotaryArgs a) {
  uint32_t t;
  int c, first;
  if (!place(a, t, c, first)) return;
  const bool turned = c < a.turned;
  const int at = turned ? 2 * c : a.pairs + c;  // behind the pairs: 2 pairs + (c - pairs)
  float2 cs = make_float2(0.f, 0.f);
  if (turned) {
    cs = cos_sin(a.positions[t], a.turns[c], a.transpose);
    cs.x *= a.factor;
    cs.y *= a.factor;
  }
  for (int h = first; h < a.all_heads; h += a.lanes) {
    const bool q = h < a.heads;
    const int g = q ? h : h - a.heads;
    const T* x = static_cast<const T*>(q ? a.q : a.k) + t * (q ? a.q_st : a.k_st) +
                 g * (q ? a.q_sh : a.k_sh) + at;
    T* y = static_cast<T*>(q ? a.q_out : a.k_out) + t * (q ? a.qo_st : a.ko_st) +
           g * (q ? a.qo_sh : a.ko_sh) + at;
    if (!turned) {
      y[0] = x[0];
      continue;
    }
    const float xa = widen(x[0]), xb = widen(x[1]);
    y[0] = narrow<T>(fmaf(xa, cs.x, -(xb * cs.y)));
    y[1] = narrow<T>(fmaf(xb, cs.x, xa * cs.y));
  }
}

// Threads that fill the GPU once.
constexpr int64_t kFull = 152 * 2048;

template <typename T, int V>
dsa_status launch(RotaryArgs a, int32_t head_dim, bool halves, cudaStream_t stream) {
  const bool pairs = !halves && V == 1;
  a.turned = halves ? a.pairs / V : pairs ? a.pairs : 2 * a.pairs / V;
  a.chunks = a.turned + (head_dim - 2 * a.pairs) / V;
  const int64_t tokens = a.tokens, units = tokens * a.chunks, want = (kFull + units - 1) / units;
  a.lanes = static_cast<uint32_t>(want < a.all_heads ? want : a.all_heads);
  // Threads of a launch are counted in 32 bits.
  const int64_t most = (INT32_MAX - kThreads) / (static_cast<int64_t>(a.chunks) * a.lanes);
  for (int64_t done = 0; done < tokens; done += most) {
    const int64_t now = tokens - done < most ? tokens - done : most;
    a.tokens = static_cast<uint32_t>(now);
    const unsigned grid =
        static_cast<unsigned>((now * a.chunks * a.lanes + kThreads - 1) / kThreads);
    if (halves)
      rotary_kernel<T, V, true><<<grid, kThreads, 0, stream>>>(a);
    else if constexpr (V == 1)
      rotary_pairs_kernel<T><<<grid, kThreads, 0, stream>>>(a);
    else
      rotary_kernel<T, V, false><<<grid, kThreads, 0, stream>>>(a);
    if (cudaGetLastError() != cudaSuccess) return DSA_ECUDA;
    a.q = static_cast<const T*>(a.q) + most * a.q_st;
    a.k = static_cast<const T*>(a.k) + most * a.k_st;
    a.q_out = static_cast<T*>(a.q_out) + most * a.qo_st;
    a.k_out = static_cast<T*>(a.k_out) + most * a.ko_st;
    a.positions += most;
  }
  return DSA_OK;
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
  if (tokens > INT32_MAX || head_dim > 65536 || all * head_dim > INT32_MAX)
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
  a.tokens = static_cast<uint32_t>(tokens);
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
